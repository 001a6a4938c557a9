"""Which form of a kernel a product takes: the launchers' rules once more, for tests that have
to reach a certain one.  RULES are the lines of the sources that they repeat: test_product_forms
looks them up, so that a rule that changes there fails here, and the sizes of the tests that
count on it are looked at again."""
import os

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "resident_expert_routing_amd", "csrc")

RULES = {
    "grouped.hpp": [
        "constexpr int kMostRows = 320;",
        "static constexpr int kCols = 64 * WA,",
        "constexpr int kSmall = 1, kLarge = 4;",
        "constexpr int kOuter = sizeof(E) == 4 ? 2 : 4;",
        "constexpr int kStep = 128;",
        "constexpr int kFewTiles = 192;",
        "constexpr int kTable = 2048;",
        "if ((M / most + groups) * cols >= 256) return most;",
        "for (int R : {320, 256, 192, 128, 64}) {",
        "const int64_t cost = ((M / R + groups) * cols + 255) / 256 * (R + 256);",
        "few = (p.M / 64 + groups) * cols;",
        "if (few < kFewTiles && (p.M <= 16 || p.M < 4 * groups)) {",
        "rows_of_tile(p.M, p.G, cols, sizeof(E) == 4 ? 128 : dma ? kMostRows : 256);",
        "const int64_t items = max_items(p.M, p.G, R) + (p.zero_rest ? 2 : 0);",
        "const bool blocks = p.M > 128 * (int64_t)p.G && items * cols >= 2048;",
        "else if (rows <= 192)\n      rows_tile<E, ACROSS, GLU, WA, 6, 2, true, false>",
        "else if (rows <= 256)\n      rows_tile<E, ACROSS, GLU, WA, 8, 2, true, false>",
        "const bool few = tiles_of(64 * WA) < kFewTiles;",
        "const bool blocks = tiles_of(side) >= 8192 && p.M >= 256 * (int64_t)p.G;",
    ],
    "int4.hip": [
        "using Few = Form<1, 2, 8, 1>;",
        "using Mid = Form<1, 2, 4, 1>;",
        "using Thin = Form<1, 4, 1, 2>;",
        "using Wide = Form<2, 4, 1, 4>;",
        "constexpr int kEnough = 640, kCUs = 256;",
        "const bool thin = p.M <= 16 || p.M < 24 * groups;",
        "if (!thin && groups * columns<Wide, GLU>(p) >= kCUs) {",
        "} else if (max_items(p.M, p.G, 16) * columns<Mid, GLU>(p) <= kCUs) {",
        "} else if (max_items(p.M, p.G, 16) * columns<Thin, GLU>(p) < kEnough) {",
    ],
    "groups.hpp": ["return (int64_t)M / R + (G > 0 ? (G < M ? G : M) : 1);"],
}

FEW = 192


def up(n, m):
    return -(-n // m)


def whole(esize, *sizes):
    """Whether rows of these lengths, in tensors of their own, are whole 16-byte pieces."""
    return all(n * esize % 16 == 0 for n in sizes)


def rows_form(M, N, G, swiglu, across, esize, dma, zero_rest=True):
    """("stream",), ("small",) or ("tiles", most rows of a tile, in XCD blocks)."""
    cols, groups = up(N, 128 if swiglu else 256), min(G, M)
    if (M // 64 + groups) * cols < FEW:
        return ("stream",) if not across and (M <= 16 or M < 4 * groups) else ("small",)
    most = 128 if esize == 4 else 320 if dma else 256
    R = most
    if (M // most + groups) * cols < 256:
        R = min((r for r in (320, 256, 192, 128, 64) if r <= most),
                key=lambda r: up((M // r + groups) * cols, 256) * (r + 256))
    items = M // R + groups + (2 if zero_rest else 0)
    return "tiles", R, M > 128 * G and items * cols >= 2048


def tile_heights(counts, R, esize, dma):
    """The heights (in sixteens of a wave's rows) of the tiles that groups of these sizes make."""
    steps = (64, 128) if esize == 4 else (64, 128, 192, 256, 320) if dma else (64, 128, 256)
    return {next(s for s in steps if min(R, n - lo) <= s) // 32
            for n in counts for lo in range(0, n, R)}


def outer_form(M, L, R, G, esize):
    """("small",) or ("tiles", in XCD blocks)."""
    side = 128 if esize == 4 else 256
    tiles = G * up(L, side) * up(R, side)
    return ("small",) if tiles < FEW else ("tiles", tiles >= 8192 and M >= 256 * G)


def int4_form(M, N, G, swiglu):
    """The form of moe_int4_matmul; G = 0: dense."""
    per = lambda cols: up(N, cols // 2 if swiglu else cols)
    groups = min(G, M) if G else 1
    items = M // 16 + groups
    thin = M <= 16 or M < 24 * groups
    if not thin and groups * per(256) >= 256:
        return "wide"
    if items * per(32) <= 256:
        return "few"
    return "mid" if items * per(128) < 640 else "thin"
