// The tiled products of grouped.hpp for bf16.
#include "grouped.hpp"

namespace moe {
template int launch_rows_product<Bf16>(const RowsProduct&, bool, bool, hipStream_t);
template int launch_outer_product<Bf16>(const OuterProduct&, hipStream_t);
}  // namespace moe
