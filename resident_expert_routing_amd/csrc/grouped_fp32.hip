// The tiled products of grouped.hpp for fp32.
#include "grouped.hpp"

namespace moe {
template int launch_rows_product<float>(const RowsProduct&, bool, bool, hipStream_t);
template int launch_outer_product<float>(const OuterProduct&, hipStream_t);
}  // namespace moe
