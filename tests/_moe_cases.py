"""Routed products that between them run every kernel of gemm_1x128_128x128_routed: the kernel that each is meant
for, the rows of each expert (T tokens of k choices, or the counts themselves) and the sizes. Codes and
scales vary from element to element where they are used."""

# kernel: "registers16", "registers32", "lds", "lds past the caches"
PRODUCT_FORMS = [
    dict(kernel="registers16", swiglu=False, counts=[3, 0, 4, 1, 0, 2], N=100, K=896),
    dict(kernel="registers16", swiglu=True, T=9, k=2, E=8, N=128, K=1280),
    dict(kernel="registers32", swiglu=False, counts=[13, 0, 32, 33, 1, 2], N=112, K=1280),
    dict(kernel="registers32", swiglu=True, T=32, k=2, E=8, N=256, K=1280),
    dict(kernel="registers32", swiglu=True, T=37, k=3, E=8, N=128, K=640, dropped=0.2),
    dict(kernel="lds", swiglu=False, counts=[70, 0, 129, 1, 64, 63], N=200, K=640),
    dict(kernel="lds", swiglu=True, T=150, k=2, E=6, N=384, K=384, dropped=0.1),
    dict(kernel="lds past the caches", swiglu=False, counts=[0, 1, 64, 65, 33] + [4] * 20 + [0, 17, 2, 90] + [1] * 9 + [3, 0], N=1272, K=512),
    dict(kernel="lds past the caches", swiglu=True, T=100, k=4, E=50, N=512, K=384),
    dict(kernel="lds past the caches", swiglu=True, T=300, k=4, E=50, N=512, K=128, dropped=0.1),
]


def rows(case):
    """M, the rows of C that a case's call has (dropped choices' and two before, three after the counts)."""
    return case["T"] * case["k"] if "T" in case else sum(case["counts"]) + 5


def experts(case):
    return case["E"] if "T" in case else len(case["counts"])
