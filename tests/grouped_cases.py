"""Grouped products that between them take every kernel, ring and tile width of the dispatch rule, and the longest walks: a CTA's
third tile meets its accumulators and its ring again.  What a case takes at 152 SMs is written beside it and checked on the CPU."""
import scaled_quantize_gemm_amax_gb300 as fq

R, O = fq.Recipe, fq.OutDtype
T, MX = R.TENSOR, R.MX_1x32_TILED
SMS = 152


def segments(experts, blocks):
    """Blocks of the experts' segments, `blocks` on the average: fewer, more, as many in turn, so some empty and some odd."""
    return [blocks + (-1, 1, 0)[e % 3] if e - e % 3 + 1 < experts else blocks for e in range(experts)]


# recipe, experts, blocks a segment, N, K | the tile's columns (0: pairs), B's stages, whether a CTA or a pair has a third tile
ROWS = [
    (T, 1, 1, 128, 1152, 32, 8, False), (T, 1, 1, 5120, 128, 64, 8, False), (T, 1, 2, 5120, 256, 96, 8, False),
    (T, 8, 8, 640, 1152, 128, 7, True), (T, 5, 1, 4096, 1024, 160, 6, False), (T, 260, 1, 640, 128, 160, 6, True),
    (T, 40, 1, 1920, 896, 192, 5, True), (T, 8, 3, 3200, 384, 224, 5, True), (T, 3, 8, 3200, 640, 256, 4, True),
    (T, 5, 3, 5120, 1152, 0, 6, True), (T, 200, 3, 256, 256, 0, 6, True), (T, 201, 3, 256, 640, 0, 5, True), (T, 260, 3, 256, 1408, 0, 5, True),
    (MX, 1, 1, 128, 1280, 64, 8, False), (MX, 8, 8, 640, 896, 128, 6, True), (MX, 5, 1, 4096, 768, 192, 5, False),
    (MX, 40, 1, 1920, 1152, 192, 5, True), (MX, 40, 1, 640, 640, 256, 4, False), (MX, 500, 1, 256, 128, 256, 4, True),
    (MX, 5, 3, 5120, 1152, 0, 5, True), (MX, 201, 2, 256, 384, 0, 5, True), (MX, 1024, 2, 256, 128, 0, 5, True),
]
# recipe, experts, blocks a segment, M, N | as above
DEPTH = [
    (T, 1, 9, 128, 128, 32, 8, False), (T, 1, 3, 128, 5120, 64, 8, False), (T, 1, 5, 256, 5120, 96, 8, False),
    (T, 40, 2, 1024, 128, 128, 7, True), (T, 5, 10, 128, 4096, 160, 6, False), (T, 260, 1, 128, 640, 160, 6, True),
    (T, 64, 2, 384, 384, 192, 5, True), (T, 40, 3, 128, 2176, 224, 5, True), (T, 40, 2, 128, 2560, 256, 4, True),
    (T, 3, 11, 1024, 3200, 0, 6, True), (T, 201, 2, 256, 256, 0, 5, True), (T, 300, 1, 384, 256, 0, 5, True),
    (MX, 1, 9, 128, 128, 64, 8, False), (MX, 40, 3, 1024, 128, 128, 6, True), (MX, 5, 9, 128, 4096, 192, 5, False),
    (MX, 64, 3, 384, 384, 192, 5, True), (MX, 40, 6, 128, 640, 256, 4, False), (MX, 500, 1, 128, 256, 256, 4, True),
    (MX, 5, 7, 384, 4096, 0, 5, True), (MX, 201, 2, 256, 256, 0, 5, True), (MX, 700, 1, 256, 256, 0, 5, True),
]


def tiles(blocks, m, n, width):
    """How many tiles a call has: m 0 for rows, whose segments have `blocks`, else of every expert's m."""
    rows = [128 * b for b in blocks] if not m else [m] * len(blocks)
    high, wide = (128, width) if width else (256, 256)
    return sum(-(-r // high) for r in rows) * -(-n // wide)
