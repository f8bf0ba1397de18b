"""The entry points with stream= given: what a call allocates for itself, and
the inputs that its caller lets go of, stay allocated until that stream has
used them, although other streams go on allocating meanwhile."""
import pytest
import torch

import ternary_quantized_linear_b200 as tql

pytestmark = pytest.mark.gpu

M, N, K = 128, 1024, 1024


def _inputs():
    g = torch.Generator(device="cuda").manual_seed(7)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    W = 0.05 * rand(N, K)
    W_packed, s_w = tql.bitnet_quantize_pack_weights(W)
    return {"x": rand(M, K), "W": W, "W_packed": W_packed, "s_w": s_w,
            "base": W.bfloat16(), "fine": (W + 0.01 * rand(N, K)).bfloat16(),
            "dy": rand(M, N).bfloat16(), "x_lam": rand(M, K).bfloat16()}


def _tensors(out):
    if isinstance(out, dict):
        out = list(out.values())
    if isinstance(out, (list, tuple)):
        return [t for t in out if t is not None]
    return [out.data if isinstance(out, tql.TiledWeights) else out]


CALLS = {
    "quantize_pack": lambda v, s: tql.bitnet_quantize_pack_weights(v("W"), stream=s),
    "quantize_pack_groups": lambda v, s: tql.bitnet_quantize_pack_weights_group_scales(
        v("W"), 256, stream=s),
    "rmsnorm_quant": lambda v, s: tql.bitnet_rmsnorm_quant_act(v("x"), stream=s),
    "forward": lambda v, s: tql.bitnet_linear_forward(v("x"), None, 1e-5, v("W_packed"),
                                                      v("s_w"), stream=s),
    "forward_ex": lambda v, s: tql.bitnet_linear_forward_ex(
        v("x"), None, 1e-5, tql.TiledWeights(tql.bitnet_tile_weights(v("W_packed")).data, N, K),
        v("s_w"), stream=s),
    "grouped": lambda v, s: tql.bitnet_linear_forward_grouped(
        ((v("x"), None, 1e-5, v("W_packed"), v("s_w"),
          torch.empty(M, N, dtype=torch.bfloat16, device="cuda")) for _ in range(2)), stream=s),
    "grouped_by_name": lambda v, s: tql.bitnet_linear_forward_grouped(
        items=((v("x"), None, 1e-5, v("W_packed"), v("s_w"),
                torch.empty(M, N, dtype=torch.bfloat16, device="cuda")) for _ in range(2)),
        stream=s),
    "tile": lambda v, s: tql.bitnet_tile_weights(v("W_packed"), None, s),
    "warmup_weights": lambda v, s: tql.bitnet_warmup_quantize_weights(v("W"), 0.5, stream=s),
    "warmup_forward": lambda v, s: tql.bitnet_warmup_forward(v("x"), None, 1e-5, v("base"), 0.5,
                                                             stream=s),
    "warmup_backward": lambda v, s: tql.bitnet_warmup_backward(v("dy"), v("x_lam"), v("base"),
                                                               stream=s),
    "bitdelta_compress": lambda v, s: tql.bitnet_bitdelta_compress(v("base"), v("fine"), stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_a_call_on_another_stream(name):
    inputs, call = _inputs(), CALLS[name]
    want = _tensors(call(lambda k: inputs[k], None))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        temporaries = {k: v.clone() for k, v in inputs.items()}
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(60_000_000)  # some 30 ms
        got = call(lambda k: temporaries[k], s)
        del temporaries
        # what the allocator hands out now on the current stream is written at once
        again = [torch.full((n,), 77, dtype=torch.uint8, device="cuda")
                 for n in (512, 4096, 1 << 15, 1 << 17, 1 << 18, 1 << 20, 1 << 21, 1 << 22)
                 for _ in range(12)]
        torch.cuda.synchronize()
        assert len(again) == 96
        assert all(torch.equal(a, b) for a, b in zip(_tensors(got), want))
