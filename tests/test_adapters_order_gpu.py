"""Calls that follow one another without a pause while what they read is written anew at the same addresses: each takes
its own plan, scales and base.  (From 33 tokens to 2048 two kernels run side by side, the second without a wait of its own
at its start; its reads go past L1, where an older line could lie.)"""
from __future__ import annotations

import os
import re

import pytest

from shared_memory_tiled_gb300 import binding as B

CSRC = os.path.join(os.path.dirname(B.__file__), "csrc")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from shared_memory_tiled_gb300 import build
    build.build()
    B.load()


def test_what_is_read_without_a_wait_is_read_past_l1():
    """k_adapters takes the plan, scale and base by __ldcg, and waits for the launch before it exactly once: at its start, or
    beside k_adapters_few at its end, which waits before it lets others start."""
    text = open(os.path.join(CSRC, "adapters.cu")).read()
    tile = text[text.index("bool plan_tile("):]
    tile = tile[:tile.index("\n}\n")]
    copy = text[text.index("void copy_rows("):]
    copy = copy[:copy.index("\n}\n")]
    many = text[text.index("\nk_adapters("):]
    many = many[:many.index("\n}\n")]
    few = text[text.index("k_adapters_few(const Few g) {"):]
    for part in (tile, copy, many):
        for access in re.findall(r"(?<!&)\*reinterpret_cast<const (?:int4|uint4) \*>\((?:plan|p \+)[^;]*;|g\.(?:plan|scale)\[[^;]*;|\? \*?p(?:\[c\])? :", part):
            raise AssertionError(access)
    assert tile.count("__ldcg(") == 2 and copy.count("__ldcg(") == 2 and many.count("__ldcg(") == 3
    assert many.count("wait_dependencies()") == 2 and "if (!g.beside) ptx::wait_dependencies();" in many
    assert many.rstrip().endswith("if (g.beside) ptx::wait_dependencies();")
    assert few.index("wait_dependencies()") < few.index("launch_dependents()") < few.index("plan_tile(")
    launch = text[text.index("cudaError_t launch_adapters("):]
    assert launch.index("launch_few_rank<16>") < launch.index("g.beside = 1") < launch.index("launch_rank<16>")


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,rank,n,out", [(20, 16, 136, "bf16"), (100, 16, 264, "bf16"), (700, 24, 265, "bf16"), (1500, 64, 264, "f32"), (2048, 8, 129, "f32"),
                                               (2100, 16, 264, "bf16")])
def test_inputs_written_anew_at_the_same_addresses(tokens, rank, n, out):
    import torch
    from test_linear_gpu import torch_types
    steps, count, k, kind = 60, 6, 136, torch_types(out)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    xs = torch.randn(steps, tokens, k, device="cuda", generator=g).bfloat16()
    bases = torch.randn(steps, tokens, n, device="cuda", generator=g).to(kind)
    scales = torch.rand(steps, count, device="cuda", generator=g) + 0.5
    # an adapter of a few tokens, those of many, and some without one
    indexes = torch.randint(-1, count - 1, (steps, tokens), device="cuda", generator=g, dtype=torch.int32)
    indexes[:, tokens // 2] = count - 1
    a = (torch.randn(count, rank, k, device="cuda", generator=g) / k ** 0.5).bfloat16()
    b = torch.randn(count, n, rank, device="cuda", generator=g).bfloat16()
    want = []
    for i in range(steps):
        want.append(B.adapters(xs[i], a, b, B.adapter_plan(indexes[i], count), scale=scales[i], base=bases[i]))
        torch.cuda.synchronize()
    x, base, scale, index = xs[0].clone(), bases[0].clone(), scales[0].clone(), indexes[0].clone()
    plan, outs = B.adapter_plan(index, count), torch.empty(steps, tokens, n, dtype=kind, device="cuda")

    def step(i):
        x.copy_(xs[i]), base.copy_(bases[i]), scale.copy_(scales[i]), index.copy_(indexes[i])
        B.check(B.tr_adapter_plan(B.AdapterPlanArgs(index=index.data_ptr(), plan=plan.words.data_ptr(), plan_bytes=plan.words.numel(), tokens=tokens,
                                                    adapters=count, stream=torch.cuda.current_stream().cuda_stream)))
        B.adapters(x, a, b, plan, scale=scale, base=base, out=outs[i])

    step(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()   # replayed without the host between the steps
    with torch.cuda.graph(graph):
        for i in range(steps):
            step(i)
    for _ in range(3):
        outs.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for i in range(steps):
            assert torch.equal(outs[i], want[i]), i
    assert B.tr_device_status() == B.Status.OK
