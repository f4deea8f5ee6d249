"""Two models alive in one process: the second's sizes must not change what the first may launch."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def run(m, s, seqs=1):
    """Prefill and three decode steps; the logits of every step."""
    from synth import make_prompt
    out = []
    for q in range(seqs):
        m.prefill(make_prompt(s, 9 + q), seq=q)
    for _ in range(3):
        m.decode_step()
        out += [m.logits(seq=q) for q in range(seqs)]
    return out


@pytest.mark.parametrize("first,cap,second,cap2,seqs", [
    ("hd128_bf16", 64, "gqa2_hd128_bf16", 64, 1),  # the persistent step kernel: a hidden vector in shared memory
    ("gqa2_hd128_bf16", 64, "hd128_bf16", 64, 1),
    ("small_f32", 8192, "small_f32", 6400, 1),     # the CUDA-core attention: a chunk of the capacity in shared memory
    ("small_f32", 6400, "small_f32", 8192, 1),
    ("small_bf16", 8192, "small_bf16", 6400, 3),   # the batched step
])
def test_a_second_model_leaves_the_first_its_launches(first, cap, second, cap2, seqs):
    from qwen2_decoder_forward_decode_gb300 import DeviceWeights, Model
    from synth import SHAPES, make_weights
    weights = {n: DeviceWeights(make_weights(SHAPES[n]), 1 if SHAPES[n].dtype == "bf16" else 0) for n in {first, second}}

    def model(name, c):
        return Model(SHAPES[name], weights[name], c, max_seqs=seqs)

    alone = []
    for name, c in ((first, cap), (second, cap2)):
        m = model(name, c)
        try:
            alone.append(run(m, SHAPES[name], seqs))
        finally:
            m.close()
    a, b = model(first, cap), model(second, cap2)
    try:
        both = [run(a, SHAPES[first], seqs), run(b, SHAPES[second], seqs)]
    finally:
        a.close()
        b.close()
    for want, got in zip(alone, both):
        for x, y in zip(want, got):
            np.testing.assert_array_equal(x, y)


class default_stream_refused:
    """A stream that waits for the default one is captured: launches on the default stream fail meanwhile."""

    def __enter__(self):
        import ctypes
        self.rt = next((ctypes.CDLL(n) for n in {line.split()[-1] for line in open("/proc/self/maps") if "libcudart.so" in line}), None)
        if self.rt is None:
            pytest.skip("no shared CUDA runtime to make a stream with")
        self.stream, self.graph = ctypes.c_void_p(), ctypes.c_void_p()
        self.byref = ctypes.byref
        assert self.rt.cudaStreamCreate(ctypes.byref(self.stream)) == 0
        assert self.rt.cudaStreamBeginCapture(self.stream, 1) == 0  # (this thread's calls only)

    def __exit__(self, *exc):
        if self.rt.cudaStreamEndCapture(self.stream, self.byref(self.graph)) == 0:  # (a failed launch ends the capture, a failed query does not)
            self.rt.cudaGraphDestroy(self.graph)
        self.rt.cudaGetLastError()
        assert self.rt.cudaStreamDestroy(self.stream) == 0


@pytest.mark.parametrize("op", ["plan", "decode attention"])
def test_a_failed_call_leaves_no_error_to_the_next(op):
    """An operator whose launch fails reports it; a model's prefill after it has none to report."""
    import test_paged_plan
    from qwen2_decoder_forward_decode_gb300 import DeviceWeights, Model, binding
    from synth import SHAPES, make_prompt, make_weights
    s = SHAPES["small_f32"]
    m = Model(s, DeviceWeights(make_weights(s), 0), 64)
    p = test_paged_plan.Plan([3, 16], [1, 1], 16, 4, 2)
    q, k, v, out = (torch.zeros(n, device="cuda") for n in (64, 32 * 16, 32 * 16, 64))
    call = {"plan": p.run, "decode attention": lambda: binding.decode_attention_noalloc(0, 4, 1, 16, 20, 32, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), None)}[op]
    torch.cuda.synchronize()
    try:
        want = m.prefill(make_prompt(s, 40))
        with default_stream_refused(), pytest.raises(binding.QwError) as e:
            call()
        assert e.value.status == 5
        assert m.prefill(make_prompt(s, 40)) == want
        call()
        p.run() if op != "plan" else p.check()
    finally:
        m.close()
