"""Sizes and types of the linear layer that between them launch every
instantiation of its kernels: (M, K, N, (x, w, output), activation), types "f"
(fp32) and "b" (bf16). test_linear_plan.py holds that they do, on the CPU;
test_gpu_linear_dispatch.py runs them."""
import itertools

TYPES = list(itertools.product("fb", repeat=3))


def large_tiles():
    """Tiles of 256 and 128: several tiles either way, ragged in rows, columns
    and reduction; rows of whole 16-byte pieces (multiples of 8) and others."""
    yield 16385, 520, 776, ("b", "b", "b"), "none"          # 256 forward
    yield 8200, 2056, 1032, ("b", "b", "b"), "none"         # 256 input gradient
    for t, K, N in itertools.product(TYPES, (1000, 1001), (264, 263)):
        yield 5200, K, N, t, "none"                         # 128 of both gradients
    for x, w, K in itertools.product("fb", "fb", (40, 44)):
        yield 4200, K, 1032, (x, w, x), "gelu"              # 128 forward; dz by a pass of its own


def small_tiles():
    """Tiles of 64: both gradients in one launch, dz as it comes or formed from
    its slope while staged; the forward pass past the few-rows kernel."""
    for t, K, N, act in itertools.product(TYPES, (72, 75), (104, 107), ("none", "silu")):
        yield 300, K, N, t, act
    for x, w, K in itertools.product("fb", "fb", (72, 75)):
        yield 700, K, 520, (x, w, x), "none"


def few_rows():
    """Every block shape of the few-rows kernel, reductions ending inside a
    piece and a round."""
    for x, w in itertools.product("fb", repeat=2):
        for M, K, N in ((7, 37, 130), (3, 65, 8200), (260, 40, 400), (100, 333, 517), (300, 600, 1100), (30, 100, 8200)):
            yield M, K, N, (x, w, "f"), "none"


def narrow():
    """The backward pass that keeps its weights in LDS, at each pair of widths."""
    for t, act in itertools.product(TYPES, ("none", "gelu")):
        for K, N in ((64, 64), (40, 104), (72, 56), (128, 72), (200, 24), (64, 256)):
            yield 66773, K, N, t, act
