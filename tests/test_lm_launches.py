"""The launches of the language-model operators, recorded on the host (lm_launches.py): their sizes, and that the GPU
tests between them launch every kernel in every way that it is used."""
import itertools
import os
import re

import pytest

import lm_launches as lm

pytestmark = pytest.mark.skipif(not os.path.exists(lm.HIPCC), reason="hipcc not installed")

MOST_ROWS, MOST_COLUMNS = 1 << 30, 1 << 21
# the largest extents that the entry points take, in each direction, and some that a card's memory holds
EXTREME_XENT = [(MOST_ROWS, 8, 1), (MOST_ROWS, 8, 128), (1 << 26, 8, 8), (1 << 24, 8, 32769), ((1 << 21) + 1, 8, 1 << 17),
                (1 << 14, MOST_COLUMNS, 512), (1, 8, MOST_COLUMNS), (1 << 12, 64, MOST_COLUMNS), (3, MOST_COLUMNS, 3)]
EXTREME_LINEAR = [(MOST_ROWS, 8, 1), (1 << 24, 8, 1 << 10), (1 << 24, 128, 1 << 14), (1, MOST_COLUMNS, MOST_COLUMNS),
                  (64, 8, MOST_COLUMNS), (1 << 14, 64, MOST_COLUMNS), (1 << 14, MOST_COLUMNS, 64)]


def fits(launches):
    assert launches
    for l in launches:
        # the runtime counts the threads along x in 32 bits, workgroups along y and z in 16
        assert 1 <= l.grid[0] and l.grid[0] * l.block[0] < 1 << 32, l
        assert 1 <= l.grid[1] < 1 << 16 and l.grid[2] == 1, l


@pytest.mark.parametrize("shape", EXTREME_XENT)
def test_launches_of_the_largest_cross_entropies_are_valid(shape):
    fits(lm.xent(*shape))
    fits(lm.xent_bwd(*shape))
    T, K, V = shape
    least = T * 512 + (T + 64) * K * 4 * 64 + (1 << 20)
    fits(lm.xent_bwd(T, K, V, work_bytes=least))


@pytest.mark.parametrize("shape", EXTREME_LINEAR)
def test_launches_of_the_largest_linear_layers_are_valid(shape):
    M, K, Nc = shape
    fits(lm.linear(M, K, Nc))
    fits(lm.linear(M, K, Nc, "silu", True, True, True))
    fits(lm.linear_bwd(M, K, Nc, "gelu"))


@pytest.mark.parametrize("shape", [(1024, 1 << 15, 64, 64), (1024, 1, 8, MOST_COLUMNS), (1, MOST_ROWS, 8, 8), (1, 1, 1 << 14, 1 << 14),
                                   (1024, 1 << 24, 64, 1 << 10)])
def test_launches_of_the_largest_grouped_products_are_valid(shape):
    fits(lm.grouped(*shape))
    fits(lm.grouped_bwd(*shape))


def test_slices_of_a_join_cover_its_rows():
    """Rows past a launch's limit go to another one, and no row to two."""
    T = MOST_ROWS
    joins = [l for l in lm.xent(T, 8, 1) if l.kernel == "xent_join<1>"]
    assert len(joins) > 1 and sum(l.grid[0] for l in joins) == T // 4
    joins = [l for l in lm.xent(1 << 24, 8, 32769) if l.kernel == "xent_join<4>"]
    assert len(joins) > 1 and sum(l.grid[0] for l in joins) == 1 << 24


class Reached:
    """What the GPU tests' calls launch: kernels, and of products also what is done with them."""

    def __init__(self):
        self.what = set()

    def add(self, launches, ends=()):
        for l in launches:
            self.what.add(l.kernel)
            if l.args is None:
                continue
            group = {0: "", 1: "grouped ", 2: "k-grouped "}[l.args.group]
            if group:
                self.what.add(group + l.kernel)
            if l.args.splits > 1:
                self.what.add("split " + l.kernel)
            if l.args.accumulate:
                self.what.add("adding " + l.kernel)
            if "256" in l.kernel:
                self.what.update("%s%s: %s" % (group, l.kernel, p) for p in lm.pieces(l, ends))


def reached_by_the_gpu_tests(tests):
    r = Reached()
    if "test_lm_ops_gpu" in tests:
        import test_lm_ops_gpu as t
        for i, (M, K, Nc) in enumerate(t.LINEAR):
            options = itertools.cycle(itertools.product(t.ACTS, (True, False), (False, True)))
            for act, b, res in itertools.islice(options, i, i + 4 * 5, 4):
                r.add(lm.linear(M, K, Nc, act, b, res, True))
        for i, (M, K, Nc) in enumerate(t.LARGE):
            r.add(lm.linear(M, K, Nc))
            r.add(lm.linear(M, K, Nc, t.ACTS[1 + i % 4], True, i % 2 == 0, True))
            r.add(lm.linear_bwd(M, Nc // 8 * 8, K))
            r.add(lm.linear_bwd(K, Nc // 8 * 8, M))
        for M, K, Nc in t.LINEAR_BWD:
            for act in t.ACTS:
                r.add(lm.linear_bwd(M, K, Nc, act))
        for sizes, spare, K, Nc in t.GROUPED:
            ends = list(itertools.accumulate(sizes))
            r.add(lm.grouped(len(sizes), ends[-1] + spare, K, Nc), ends)
            r.add(lm.grouped_bwd(len(sizes), ends[-1] + spare, K, Nc), ends)
        for T, K, V in t.XENT:
            r.add(lm.xent(T, K, V))
            r.add(lm.xent_bwd(T, K, V))
            if T <= 300:
                r.add(lm.xent_bwd(T, K, V, work_bytes=1 << 20))
        for n in (900 << 10, 1200 << 10):
            r.add(lm.xent_bwd(300, 264, 3001, work_bytes=n))
    if "test_lm_kernels_gpu" in tests:
        import test_lm_kernels_gpu as t
        for case in t.LINEAR + [(4353, 1000, 4091, "gelu", True, True, True)]:
            r.add(lm.linear(*case))
        for case in t.LINEAR_BWD:
            r.add(lm.linear_bwd(*case))
        for cases, call in ((t.GROUPED_FWD + t.GROUPED_FEW, lm.grouped), (t.GROUPED_BWD + t.GROUPED_FEW, lm.grouped_bwd)):
            for sizes, spare, K, Nc in cases:
                ends = list(itertools.accumulate(sizes))
                r.add(call(len(sizes), ends[-1] + spare, K, Nc), ends)
        for case in t.XENT:
            r.add(lm.xent(*case))
            r.add(lm.xent_bwd(*case))
        for case in t.XENT_PIECES:
            r.add(lm.xent_bwd(*case))
    return r.what


GPU_TESTS = ("test_lm_ops_gpu", "test_lm_kernels_gpu")


def test_every_kernel_is_launched_by_a_gpu_test():
    """The shapes of the GPU tests go where the plans send them: a changed plan that leaves a kernel to no test fails
    here, and so does a kernel that no call reaches."""
    missing = lm.kernels() - reached_by_the_gpu_tests(GPU_TESTS)
    assert not missing, sorted(missing)


def test_every_use_of_a_product_is_launched_by_a_gpu_test():
    cuts = ["tile", "half of tile", "lone half", "quarter of tile", "lone quarter"]
    want = ["%s: %s" % (k, c) for k in ("nt256<0>", "nt256<1>", "nt256<2>", "nt256<3>", "nn256", "tn256") for c in cuts]
    want += ["grouped %s: %s" % (k, c) for k in ("nt256<3>", "nn256")
             for c in cuts + ["pair", "half of pair", "quarter of pair"]]
    want += ["k-grouped tn256: " + c for c in ("tile", "lone half")]
    want += ["grouped " + k for k in ("nt128<3>", "nn128", "nn32", "rows<1,4,0>", "rows<1,8,0>", "rows<2,4,0>", "rows<2,6,0>",
                                      "rows_wide<1,0>", "rows_wide<2,0>")] + ["k-grouped tn128"]
    want += ["split " + k for k in ("nt128<3>", "nn256", "nn128", "nn32", "tn128")]
    want += ["adding " + k for k in ("nn256", "nn128", "nnshort", "nn32")]
    missing = set(want) - reached_by_the_gpu_tests(GPU_TESTS)
    assert not missing, sorted(missing)


def logits_kernel(T, K, V):
    return lm.xent(T, K, V)[0].kernel


def test_logits_of_few_tiles_go_to_the_few_rows_kernel():
    """By the number of its tiles and the reduction's length alone, in the backward pass as in the forward one."""
    for T, V in ((65, 1), (384, 1003), (1024, 500), (2048, 500), (4096, 200), (16384, 64), (512, 2048)):
        for K in (8, 256, 576, 4096):
            assert logits_kernel(T, K, V) == "rows_wide<4,1>", (T, K, V)
            assert lm.xent_bwd(T, K, V)[0].kernel == "rows_wide<4,2>", (T, K, V)
    for T, V in ((200, 8000), (1024, 2048), (384, 4427)):        # up to two tiles for a CU
        assert logits_kernel(T, 1024, V) == "rows_wide<4,1>"
        assert logits_kernel(T, 1032, V) == "nt128<1>"
    for T, V in ((1024, 2049), (8192, 300), (65, 1 << 20)):
        assert not logits_kernel(T, 8, V).startswith("rows")


def test_many_groups_of_a_short_reduction_go_to_tiles():
    """Whatever the skew: all rows of 1024 groups may be one group's."""
    few = lambda E, M, K, Nc: lm.grouped(E, M, K, Nc)[0].kernel.startswith("rows")
    for E, K in ((1024, 512), (1024, 8184), (65, 512), (129, 1024), (256, 2040)):
        for rows in (1, E, 32 * E):
            assert not few(E, rows, K, 512), (E, K, rows)
    for E, K in ((1, 8), (64, 8), (64, 512), (128, 1024), (1024, 8192)):
        assert few(E, 1, K, 512) and few(E, 33 * E - 1, K, 512) and not few(E, 33 * E, K, 512), (E, K)


def test_gradients_of_experts_weights_take_the_tallest_tiles_from_a_round_of_them_on():
    for E, M, K, Nc in ((8, 8000, 1024, 1024), (4, 64, 1024, 1024), (100, 100, 256, 256), (1, 5000, 512, 512), (255, 255, 8, 8)):
        assert lm.grouped_bwd(E, M, K, Nc)[1].kernel == "tn128", (E, K, Nc)
    for E, M, K, Nc in ((16, 16, 1024, 1024), (8, 8000, 2048, 2048), (256, 300, 8, 8)):
        assert lm.grouped_bwd(E, M, K, Nc)[1].kernel == "tn256", (E, K, Nc)


def test_long_reductions_of_few_rows_are_split_over_tiles():
    few = lambda M, K, Nc: lm.linear(M, K, Nc)[0].kernel.startswith("rows")
    for M, K, Nc in ((1, 32768, 97), (16, 8192, 1000), (32, 4096, 97), (64, 2048, 2000), (17, 16384, 4600), (64, 4096, 7000),
                     (64, 16384, 10000), (1, 8192, 8192), (65, 64, 64)):
        assert not few(M, K, Nc), (M, K, Nc)
    for M, K, Nc in ((1, 4096, 4096), (1, 16384, 97), (16, 4096, 1000), (32, 2048, 97), (64, 1024, 2000), (32, 4096, 4600),
                     (64, 2048, 7000), (48, 4096, 14336), (64, 16384, 14336), (1, 4096, 8192), (64, 8, 1)):
        assert few(M, K, Nc), (M, K, Nc)


@pytest.mark.parametrize("T,V,K", [(1, 1, 8), (33, 50257, 1024), (4096, 65536, 64), (4096, 65537, 64), (4096, 50257, 2048),
                                   (8192, 32769, 128), (8192, 128256, 4096), (8192, 1 << 20, 4096), (1 << 20, 257, 1024),
                                   (1 << 20, 1 << 17, 1024), (1 << 22, 600, 64)])
def test_workspace_of_the_gradient_is_a_piece_of_d_logits_and_the_sums_of_dA(T, V, K):
    """To the byte: pieces of at most 512 MiB (256 columns where that is more), in as few as that takes, and the fp32 sums
    that the launches write."""
    launches = lm.xent_bwd(T, K, V)
    logits = [l for l in launches if l.args and l.args.K == K and l.args.M == T and not l.args.part and "<" in l.kernel]
    dA = [l for l in launches if l.kernel.startswith("nn")]
    pieces, most = len(logits), max(256, (512 << 20) // (2 * T) // 256 * 256)
    assert sum(l.args.N for l in logits) == V and pieces == -(-V // most) == len(dA)
    piece = -(-(-(-V // pieces)) // 256) * 256
    assert piece <= most and all(l.args.N == piece for l in logits[:-1])
    splits = dA[0].args.splits
    assert all(l.args.splits == splits and l.args.part == (pieces > 1 or splits > 1) for l in dA)
    assert [l.args.accumulate for l in dA] == [0] + [1] * (pieces - 1)
    region = lambda n: -(-n // 256) * 256
    want = region(T * piece * 2) + (region(splits * T * K * 4) if pieces > 1 or splits > 1 else 0)
    assert lm.recorder().gemm_xent_bwd_workspace(T, V, K) == want
    # an eighth of that is enough where it holds the narrowest piece, and then only makes more of them
    least = region(T * 512) + region(64 * T * K * 4)
    if want // 8 >= least:
        assert len([l for l in lm.xent_bwd(T, K, V, work_bytes=want // 8) if l.kernel.startswith("nn")]) > pieces


def test_nothing_is_declared_that_nothing_uses():
    """Functions, constants and enumerators that the operators' files share each stand in a use outside their declaration."""
    csrc = os.path.join(lm.ROOT, "allgather_gemm_amd", "csrc")
    text = {f: re.sub(r"//.*", "", open(os.path.join(csrc, f), encoding="utf-8").read())
            for f in os.listdir(csrc) if f.startswith("lm_")}
    shared = text["lm_internal.hpp"]
    functions = re.findall(r"^(?:int|int64_t|hipError_t) (\w+)\(", shared, re.M)
    constants = re.findall(r"constexpr \w+ (\w+) =", shared) + re.findall(r"\b(k\w+) = \d", shared)
    assert len(functions) > 8 and len(constants) > 12
    code = "\n".join(text.values())
    for f in functions:                # neither declared nor defined there, but called
        assert re.search(r"(?<!^int )(?<!^int64_t )(?<!^hipError_t )\b%s\(" % f, code, re.M), f
    for c in constants:
        assert any(re.search(r"\b%s\b" % c, text[f]) for f in text if f != "lm_internal.hpp"), c
