"""Products of language models at sizes that the rules give to each tile edge, whole tiles and edges of them.
`kernel` is the one that the case is there for; `pitch` is "lines" for outputs whose rows are whole 128-byte
lines (whole tiles are then stored past the caches) and "odd" for rows that are not."""


def forward(m, n, k, t, out, ta, tb, act, kernel, bias=None, aux=False, beta=0.0, c=None, in_place=False, pitch="lines"):
    return dict(locals())


def slope(m, n, k, t, out, ta, tb, act, kernel, dbias=True, pitch="lines"):
    return dict(locals())


def grouped(rows, groups, n, k, t, out, tb, act, kernel, division, bias=False, aux=False, pitch="lines"):
    return dict(locals())


def wgrad(groups, rows, m, n, t, out, kernel, division, beta=0.0, pitch="lines"):
    return dict(locals())


def cross_entropy(m, n, k, t, kernels, train=True, ignored="some"):
    return dict(locals())


def few(m, n, k, tb, kernel, groups=0):
    """A product of few rows (of `groups` experts, where there are any)."""
    return dict(locals())


T64, T128, T256 = ("tile", 64), ("tile", 128), ("tile", 256)

FORWARD = [
    forward(300, 520, 136, "bf16", "bf16", False, True, "silu", T64, bias="bf16", aux=True, beta=1.0, c="bf16"),
    forward(200, 520, 136, "f16", "f16", True, False, "none", T64),
    forward(330, 456, 72, "f16", "f32", False, False, "gelu", T64, beta=-0.5, c="f32"),
    forward(2600, 2504, 136, "bf16", "bf16", False, True, "gelu", T128, bias="bf16", aux=True),
    forward(2600, 2504, 136, "f16", "f16", True, True, "silu", T128, bias="f32", aux=True, beta=1.0, c="f16", pitch="odd"),
    forward(2600, 2504, 72, "bf16", "f32", True, False, "relu", T128, bias="bf16", beta=0.5, c="f32", in_place=True),
    forward(2500, 2600, 72, "f16", "f16", False, False, "none", T128, beta=2.0, c="f32"),
    forward(3000, 3000, 1300, "bf16", "bf16", False, True, "silu", T256, bias="bf16", aux=True, beta=1.0, c="bf16"),
    forward(3000, 2936, 1203, "bf16", "bf16", False, True, "gelu", T256, bias="bf16", aux=True),
    forward(2936, 3000, 1200, "f16", "f32", False, False, "gelu_tanh", T256, bias="f16", beta=0.5, c="f32"),
    forward(2936, 3000, 600, "bf16", "bf16", True, False, "none", T256),
    forward(2100, 4040, 1600, "f16", "f16", True, True, "gelu", T256, bias="f32", aux=True, beta=-0.5, c="f32", pitch="odd"),
    forward(4040, 2104, 1200, "f16", "f32", False, True, "none", T256, beta=1.0, c="f32", in_place=True),
    forward(4040, 2104, 1300, "bf16", "f32", True, True, "relu", T256, bias="bf16", aux=True, beta=1.0, c="bf16", pitch="odd"),
]
SLOPE = [
    slope(300, 520, 136, "bf16", "bf16", False, True, "gelu", T64),
    slope(2600, 2504, 136, "f16", "f16", False, True, "relu", T128),
    slope(2600, 2504, 136, "bf16", "f32", True, False, "gelu_tanh", T128, pitch="odd"),
    slope(3000, 3000, 1100, "f16", "f16", False, True, "gelu_tanh", T256),
    slope(3000, 2936, 900, "bf16", "bf16", False, False, "silu", T256),
    slope(2104, 4040, 1203, "bf16", "f32", True, True, "gelu", T256, pitch="odd"),
    slope(4040, 2104, 600, "bf16", "bf16", True, False, "none", T256, dbias=False),
]
GROUPED = [
    grouped(2000, 5, 1500, 500, "bf16", "bf16", True, "silu", T64, "gaps", bias=True, aux=True),
    grouped(1999, 7, 1490, 1003, "f16", "f32", False, "none", T128, "even", bias=True),
    grouped(3000, 4, 2504, 1000, "bf16", "bf16", True, "silu", T128, "gaps", bias=True, aux=True),
    grouped(3000, 4, 2504, 1000, "f16", "f16", False, "gelu", T128, "one has all", pitch="odd"),
    grouped(4000, 6, 2904, 1200, "bf16", "bf16", True, "silu", T256, "gaps", bias=True, aux=True),
    grouped(5000, 4, 2104, 1500, "f16", "f16", False, "gelu_tanh", T256, "even"),
    grouped(5000, 4, 2104, 1500, "bf16", "f32", True, "none", T256, "single rows", aux=True, pitch="odd"),
]
GROUPED_GRAD = [
    grouped(3000, 4, 2504, 1000, "bf16", "bf16", True, "silu", T128, "even"),
    grouped(1999, 7, 1490, 1003, "f16", "f32", False, "gelu_tanh", T128, "gaps"),
    grouped(5000, 4, 2104, 1500, "bf16", "bf16", False, "silu", T256, "gaps"),
    grouped(4000, 6, 2904, 1200, "f16", "f16", True, "relu", T256, "single rows", pitch="odd"),
]
WGRAD = [
    wgrad(3, 700, 1304, 1200, "bf16", "bf16", T128, "gaps"),
    wgrad(3, 2100, 1500, 2008, "bf16", "bf16", T256, "gaps"),
    wgrad(3, 2100, 1500, 2000, "f16", "f16", T256, "one has all", beta=0.5, pitch="odd"),
    wgrad(6, 3000, 1304, 1500, "bf16", "f32", T256, "even", beta=1.0),
]
CE = [
    cross_entropy(2047, 5021, 1000, "f16", dict(logits=T256), train=False),
    cross_entropy(2500, 4104, 136, "bf16", dict(logits=T128), train=False, ignored="none"),
    cross_entropy(1000, 9000, 3000, "bf16", dict(logits=T256, dw=T256, dx=T256, splits=5)),
    cross_entropy(1030, 8903, 2500, "f16", dict(logits=T256, dw=T128, dx=T256, splits=5), ignored="none"),
    cross_entropy(700, 9000, 3000, "f16", dict(logits=T128, dw=T256, dx=T128, splits=3)),
]

# n = 2^15, so that a row's probabilities of equal logits are a power of two; two pieces of the vocabulary
PIECES = [
    cross_entropy(4096, 32768, 2048, "bf16", dict(logits=T256, dw=T256, dx=T256, splits=2, pieces=2)),
    cross_entropy(4096, 32768, 4096, "f16", dict(logits=T256, dw=T256, dx=T256, splits=1, pieces=2)),
]

# every kernel for few rows: ("few", row blocks of 16, column blocks of 16, waves)
FEW = [
    few(3, 520, 300, True, ("few", 1, 1, 8)), few(16, 9001, 203, True, ("few", 1, 1, 4)),
    few(13, 24603, 300, True, ("few", 1, 4, 4)), few(20, 523, 1030, True, ("few", 2, 2, 8)),
    few(29, 16501, 203, True, ("few", 2, 2, 4)), few(50, 1003, 300, True, ("few", 4, 2, 8)),
    few(7, 523, 300, False, ("few", 1, 2, 8)), few(15, 16501, 203, False, ("few", 1, 2, 4)),
    few(17, 523, 1030, False, ("few", 2, 2, 8)), few(32, 16501, 203, False, ("few", 2, 2, 4)),
    few(64, 1003, 300, False, ("few", 4, 2, 8)),
]
FEW_OF_EXPERTS = [
    few(50, 203, 300, True, ("few", 1, 1, 8), groups=20), few(200, 1003, 203, True, ("few", 1, 1, 4), groups=40),
    few(280, 1003, 203, True, ("few", 1, 4, 4), groups=40), few(200, 203, 300, True, ("few", 2, 2, 8), groups=9),
    few(50, 203, 300, False, ("few", 1, 2, 8), groups=20), few(200, 555, 203, False, ("few", 1, 2, 4), groups=40),
    few(200, 1003, 203, False, ("few", 1, 4, 4), groups=40), few(200, 203, 300, False, ("few", 2, 2, 8), groups=9),
]
