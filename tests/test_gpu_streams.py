"""Calls on a stream that is not the current one: their outputs are no memory
that the current stream still writes."""
from types import SimpleNamespace

import pytest

from helpers import slot_inputs, to_dev, weights
from nvfp4_gated_deltanet_gb300 import synth

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def overlap(a, b):
    return a.data_ptr() < b[1] and b[0] < a.data_ptr() + a.numel() * a.element_size()


@pytest.mark.parametrize("duck", [False, True])
@pytest.mark.parametrize("which", ["quantize", "gemm", "kda", "decode", "mix", "in_proj", "in_mix", "out_proj", "verify",
                                   "prefill"])
def test_outputs_for_a_stream_are_no_memory_that_another_still_writes(which, duck):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_gated_deltanet_gb300 as pkg
    sh = synth.FULL
    gen = torch.Generator(device="cuda").manual_seed(1)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    x = rand(64, sh.hidden).bfloat16()
    codes, scales = pkg.nvfp4_quantize(x, 0.01)
    kda = [rand(2, 4, 128) * 0.1 for _ in range(3)] + [-rand(2, 4, 128).abs(), rand(2, 4).sigmoid(), rand(2, 4, 128, 128)]
    layer = pkg.layer_from_synth(weights("FULL", 1), max_batch=16, max_prefill_tokens=64)
    _, conv0, ssm0 = slot_inputs(sh, [0, 1], 1)
    conv0, ssm0 = to_dev(conv0), to_dev(ssm0)
    ids = torch.arange(2, dtype=torch.int32, device="cuda")
    bits = x.view(torch.int16)
    proj = layer.in_proj(bits[:2].contiguous(), ids)
    mixed = layer.in_mix(bits[:2].contiguous(), ids, conv0.clone(), ssm0.clone())
    nq = proj.shape[1] - 2 * sh.n_v_heads
    qkvz, ba = proj[:, :nq].contiguous(), proj[:, nq:].contiguous()
    snaps = layer.new_snapshots(2, 2)
    rows2, rows22 = bits[:2].contiguous(), bits[:4].reshape(2, 2, -1).contiguous()
    conv, ssm, state = conv0.clone(), ssm0.clone(), kda[5].clone()

    def call(stream=None):
        calls = {
            "quantize": lambda: pkg.nvfp4_quantize(x, 0.01, stream=stream),
            "gemm": lambda: (pkg.nvfp4_gemm(codes, scales, 0.01, codes, scales, 0.01, stream=stream),),
            "kda": lambda: (pkg.kda_step(*kda[:5], state, stream=stream),),
            "decode": lambda: (layer.decode_step(rows2, ids, conv, ssm, stream=stream),),
            "mix": lambda: (layer.mix_step(qkvz, ba, ids, conv, ssm, stream=stream),),
            "in_proj": lambda: (layer.in_proj(rows2, ids, stream=stream),),
            "in_mix": lambda: layer.in_mix(rows2, ids, conv, ssm, stream=stream),
            "out_proj": lambda: (layer.out_proj(*mixed, stream=stream),),
            "verify": lambda: (layer.verify(rows22, ids, conv, ssm, *snaps, stream=stream),),
            "prefill": lambda: (layer.prefill(bits, 0, True, conv, ssm, stream=stream),)}
        return calls[which]()

    def fresh():
        conv.copy_(conv0)
        ssm.copy_(ssm0)
        state.copy_(kda[5])

    fresh()
    want = [y.clone() for y in call()]
    big = rand(4096, 4096).bfloat16()
    real = torch.cuda.Stream()
    side = SimpleNamespace(cuda_stream=real.cuda_stream) if duck else real
    for _ in range(3):
        fresh()
        torch.cuda.synchronize()
        held = [torch.empty_like(y) for y in want for _ in range(4)]
        for _ in range(20):
            big @ big
        for y in held:
            y.fill_(7)
        at = [(y.data_ptr(), y.data_ptr() + y.numel() * y.element_size()) for y in held]
        del held, y
        got = call(side)
        assert not any(overlap(y, b) for y in got for b in at)
        torch.cuda.synchronize()
        assert layer.check() == 0 and all(torch.equal(p, q) for p, q in zip(got, want))
        del got
