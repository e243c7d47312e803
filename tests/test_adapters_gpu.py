"""Low-rank adapters of many requests on the GPU: the plan against a stable sort, the outputs against
their 64-bit form."""
from __future__ import annotations

import numpy as np
import pytest

import norm_ref as N
from shared_memory_tiled_gb300 import binding as B
from test_linear_gpu import close, host, torch_types

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from shared_memory_tiled_gb300 import build
    build.build()
    B.load()
    assert B.tr_device_status() == B.Status.OK
    yield
    assert B.tr_device_status() == B.Status.OK


def words(plan):
    import torch
    return plan.words.view(torch.int32).cpu().numpy()


@pytest.mark.parametrize("tokens,count", [(1, 1), (1, 0), (31, 3), (33, 1), (64, 48), (129, 2), (1000, 7), (5000, 1), (3000, 2000), (700, 32767),
                                          (40000, 300)])
def test_plan_is_a_stable_sort(tokens, count):
    import torch
    rng = np.random.default_rng(tokens + count)
    index = rng.integers(-1, count + 1, tokens).astype(np.int32)  # -1 and `count` have none
    if tokens > 500:
        index[100:400] = index[100]
        index[rng.integers(0, tokens, 20)] = [-2 ** 31, 2 ** 31 - 1] * 10
    w = words(B.adapter_plan(torch.from_numpy(index).cuda(), count))
    group = np.where((index < 0) | (index >= count), count, index)
    large, small, order = w[0], w[3], w[-tokens:]
    assert w[1] == tokens and w[2] == count
    assert np.array_equal(order, np.argsort(group, kind="stable"))
    want, at = [[], []], 0
    for g in range(count + 1):
        n = int((group == g).sum())
        for k in range(0, n, 128):
            want[min(128, n - k) <= 16].append((g, at + k, min(128, n - k), 0))
        at += n
    table = w[4:-tokens].reshape(-1, 4)
    assert large == len(want[0]) and small == len(want[1]) and large + small <= len(table)
    assert np.array_equal(table[:large], np.array(want[0]).reshape(-1, 4))
    assert np.array_equal(table[::-1][:small], np.array(want[1]).reshape(-1, 4))


def held(values, pitch, shape_off=0):
    """bf16 on the GPU with a row pitch of its own, a sentinel between the rows."""
    import torch
    t = torch.from_numpy(values.astype(np.float32)).bfloat16()
    buf = torch.full((*values.shape[:-1], pitch), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = buf[..., :values.shape[-1]]
    v.copy_(t)
    return v, t.to(torch.float64).numpy()


def up8(n):
    return -(-n // 8) * 8


def problem(tokens, count, k, n, rank, seed, out="bf16", index=None, pitch=0):
    import torch
    rng = np.random.default_rng(seed)
    x, wx = held(rng.standard_normal((tokens, k)) * np.exp(0.5 * rng.standard_normal((tokens, 1))), up8(k) + pitch)
    a, wa = held(rng.standard_normal((count, rank, k)) / max(k, 1) ** 0.5, up8(k) + pitch)
    b, wb = held(rng.standard_normal((count, n, rank)), up8(rank) + pitch)
    scale = rng.random(count).astype(np.float32) + 0.5
    if index is None:
        index = rng.integers(-1, count, tokens)
    index = np.asarray(index, np.int32)
    base = torch.from_numpy(rng.standard_normal((tokens, n)).astype(np.float32)).to(torch_types(out)).cuda()
    return dict(x=x, a=a, b=b, scale=torch.from_numpy(scale).cuda(), plan=B.adapter_plan(torch.from_numpy(index).cuda(), count), base=base), \
        (wx, wa, wb, scale, index)


def check(p, w, out, got, base="base"):
    want, bound = N.adapters(*w, None if base is None else host(p["base"]))
    close(host(got), want, bound, out)


# tokens, adapters, k, n, rank: single tokens, tiles that end anywhere, a contraction and columns of
# one value, of less than a tile and of more than one CTA's part, ranks from 1 to 128, both sides of each kernel's limit
CASES = [(1, 1, 8, 8, 8), (1, 3, 1, 1, 1), (2, 1, 64, 128, 16), (5, 4, 100, 77, 5), (17, 3, 1111, 129, 12), (64, 48, 520, 300, 16),
         (128, 1, 512, 256, 32), (129, 2, 513, 257, 64), (300, 5, 1000, 1000, 128), (200, 2, 4096, 96, 100), (77, 9, 64, 2049, 33),
         (1000, 3, 264, 520, 8), (260, 1, 8192, 24, 127), (400, 30, 136, 4096, 24), (32, 1, 300, 200, 16), (33, 1, 300, 200, 16), (2048, 90, 72, 136, 16),
         (2049, 90, 72, 136, 16), (2300, 2, 1032, 264, 64), (20000, 3, 40, 72, 32), (64, 2, 520, 301, 12), (65, 2, 300, 200, 16),
         (32, 1, 300, 200, 17), (64, 2, 300, 200, 17), (400, 3, 2100, 1153, 40)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES)
def test_adapters(case, out):
    import torch
    p, w = problem(*case, seed=sum(case), out=out)
    got = B.adapters(p["x"], p["a"], p["b"], p["plan"], scale=p["scale"], base=p["base"])
    check(p, w, out, got)
    again = B.adapters(p["x"], p["a"], p["b"], p["plan"], scale=p["scale"], base=p["base"])
    assert torch.equal(got, again)
    bare = torch.from_numpy(w[4] < 0).cuda()
    assert torch.equal(got[bare], p["base"][bare])
    inside = p["base"].clone()  # in base's place
    assert B.adapters(p["x"], p["a"], p["b"], p["plan"], scale=p["scale"], base=inside, out=inside) is inside
    assert torch.equal(inside, got)


@pytest.mark.parametrize("n", [264, 265])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_prompts_in_turn(out, n):
    """Adapters whose requests do not lie side by side: tiles that begin, go on and end inside runs of tokens."""
    runs = [50, 94, 222, 37, 31, 128, 300, 1, 33, 2, 64, 97, 160, 5]
    for k, order in ((72, [0, 1] * 7), (1040, [2, 0, 1, 0, -1, 0, 1, 2, 0, 0, 2, 1, 0, 2])):
        p, w = problem(sum(runs), 3, k, n, 24, len(runs) + k, out, index=np.repeat(order, runs))
        check(p, w, out, B.adapters(p["x"], p["a"], p["b"], p["plan"], scale=p["scale"], base=p["base"]))


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_without_base_and_scale(out):
    import torch
    p, w = problem(150, 3, 200, 130, 20, 3, out)
    got = B.adapters(p["x"], p["a"], p["b"], p["plan"], out_dtype=torch_types(out))
    check(p, (*w[:3], np.ones(3), w[4]), out, got, None)
    assert bool((got[torch.from_numpy(w[4] < 0).cuda()] == 0).all())


def test_pitches_and_what_lies_beside():
    """Operands with room between their rows, an output that starts anywhere: nothing beside it is written."""
    import torch
    for out, pitch, off in [("bf16", 131, 1), ("f32", 131, 3), ("bf16", 136, 8), ("f32", 132, 4), ("bf16", 132, 4)]:
        p, w = problem(140, 3, 200, 130, 20, 4, out, pitch=16)
        buf = torch.full((off + 140 * pitch + 16,), 7.0, dtype=torch_types(out), device="cuda")
        view = buf[off:off + 140 * pitch].view(140, pitch)[:, :130]
        got = B.adapters(p["x"], p["a"], p["b"], p["plan"], scale=p["scale"], base=p["base"], out=view)
        check(p, w, out, got)
        assert bool((buf[:off] == 7).all()) and bool((buf[off + 140 * pitch:] == 7).all())
        assert bool((buf[off:off + 140 * pitch].view(140, pitch)[:, 130:] == 7).all())


def test_everybody_bare_and_indexes_out_of_range():
    import torch
    index = np.array([-1, 5, 2 ** 31 - 1, -2 ** 31, 3] * 30)
    p, w = problem(150, 3, 64, 100, 16, 5, index=index)
    assert torch.equal(B.adapters(p["x"], p["a"], p["b"], p["plan"], base=p["base"]), p["base"])
    p["plan"] = B.adapter_plan(torch.zeros(150, dtype=torch.int32, device="cuda"), 0)
    assert torch.equal(B.adapters(p["x"], p["a"][:0], p["b"][:0], p["plan"], base=p["base"]), p["base"])


def test_nan_stays_with_its_token_and_its_adapter():
    import torch
    index = np.arange(150) % 3
    p, w = problem(150, 3, 264, 140, 16, 6, index=index)
    clean = B.adapters(p["x"], p["a"], p["b"], p["plan"], base=p["base"])
    p["x"][7, 3], p["x"][9, 100] = float("nan"), float("inf")
    got = B.adapters(p["x"], p["a"], p["b"], p["plan"], base=p["base"])
    assert bool(got[7].isnan().all()) and not bool(got[9].isfinite().any())
    keep = [i for i in range(150) if i not in (7, 9)]
    assert torch.equal(got[keep], clean[keep])
    p["a"][1] = float("nan")
    got = B.adapters(p["x"], p["a"], p["b"], p["plan"], base=p["base"])
    keep = [i for i in keep if i % 3 != 1]
    assert torch.equal(got[keep], clean[keep]) and bool(got[1].isnan().all())


def test_nothing_to_do():
    import torch
    p, w = problem(20, 2, 40, 30, 8, 7)
    none = B.adapters(p["x"][:0], p["a"], p["b"], B.adapter_plan(torch.empty(0, dtype=torch.int32, device="cuda"), 2))
    assert none.shape == (0, 30)
    assert B.adapters(p["x"], p["a"], p["b"][:, :0], p["plan"]).shape == (20, 0)
    # no contraction: base as it is
    assert torch.equal(B.adapters(p["x"][:, :0], p["a"][:, :, :0], p["b"], p["plan"], base=p["base"]), p["base"])


def test_other_stream_and_two_graphs():
    """One batch's plan serves two projections; graphs replayed in turn share no memory of the library's."""
    import torch
    graphs, kept = [], []
    for seed in (8, 9):
        p, w = problem(90, 4, 520, 300, 16, seed)
        index = torch.from_numpy(w[4]).cuda()

        def step(p=p, index=index, stream=None):
            plan = B.adapter_plan(index, 4, stream=stream)
            first = B.adapters(p["x"], p["a"], p["b"], plan, scale=p["scale"], base=p["base"], stream=stream)
            return first, B.adapters(p["x"], p["a"], p["b"], plan, base=first, stream=stream)

        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append(g)
        kept.append((p, index, out, step))
    for p, index, _, _ in kept:
        p["x"].normal_()
        index.copy_(torch.randint(-1, 4, (90,), device="cuda"))
    for g in (graphs[1], graphs[0], graphs[1]):
        g.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for p, index, out, step in kept:
        eager = step(stream=side.cuda_stream)
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    """Calls that run side by side: each stream's answers are those of the same calls one after another."""
    import torch
    jobs = [problem(tokens, 6, 1032, 1544, rank, seed)[0] for tokens, rank, seed in ((40, 16, 1), (700, 64, 2), (2300, 32, 3), (90, 128, 4))]

    def all_of(streams):
        outs = []
        for turn in range(4):
            for i, p in enumerate(jobs):
                st = streams[(i + turn) % len(streams)]
                with torch.cuda.stream(st):
                    outs.append(B.adapters(p["x"], p["a"], p["b"], p["plan"], scale=p["scale"], base=p["base"]))
        torch.cuda.synchronize()
        return outs

    torch.cuda.synchronize()
    alone = all_of([torch.cuda.current_stream()])
    for a, b in zip(alone, all_of([torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.Stream()])):
        assert torch.equal(a, b)


def test_refusals():
    import torch
    p, w = problem(20, 2, 40, 30, 8, 10)
    x, a, b, plan = p["x"], p["a"], p["b"], p["plan"]
    with pytest.raises(TypeError):
        B.adapter_plan(torch.zeros(5, dtype=torch.int64, device="cuda"), 2)
    with pytest.raises(ValueError):
        B.adapter_plan(torch.zeros(5, dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        B.adapter_plan(torch.zeros(10, dtype=torch.int32, device="cuda")[::2], 2)
    for count in (-1, 1 << 15):
        with pytest.raises(ValueError):
            B.adapter_plan(torch.zeros(5, dtype=torch.int32, device="cuda"), count)
    with pytest.raises(TypeError):
        B.adapters(x.float(), a, b, plan)
    with pytest.raises(ValueError):
        B.adapters(x[:19], a, b, plan)
    with pytest.raises(ValueError):
        B.adapters(x, a[:1], b, plan)
    with pytest.raises(ValueError):
        B.adapters(x, a, b[:, :, :7], plan)
    with pytest.raises(ValueError):
        B.adapters(x, a, b, plan, base=p["base"][:, :29])
    with pytest.raises(TypeError):
        B.adapters(x, a, b, plan, base=p["base"], out_dtype=torch.float32)
    with pytest.raises(ValueError):
        B.adapters(x, a, b, plan, scale=p["scale"][:1])
    big = torch.zeros(1, 200, 40, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 30, 200, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(B.TransposeError):
        B.adapters(x, *big, B.adapter_plan(torch.zeros(20, dtype=torch.int32, device="cuda"), 1))
    with pytest.raises(B.TransposeError):  # rows off 16-byte boundaries
        B.adapters(torch.zeros(20, 41, dtype=torch.bfloat16, device="cuda")[:, :40], a, b, plan)
    with pytest.raises(B.TransposeError):
        B.adapters(x, a, b, plan, out=x[:, :30])
