"""The division of the GPU between the two kernels of attention over a common prefix, where calls take from some 0.4 ms to
several ms: more keys in common are more work for the kernel that takes them, and do not get it fewer SMs."""
import pytest
import torch

pytestmark = pytest.mark.gpu
PAGE, DIM, OWN = 16, 128, 64                                           # each sequence has 64 positions of its own


class Shared:
    """One group of sequences on a prefix of up to `most` positions, `new` tokens of each."""

    def __init__(self, w, seqs, new, heads, kv_heads, most):
        g = torch.Generator(device="cuda").manual_seed(seqs + heads)
        self.w, self.seqs, self.new, self.heads, self.kv_heads, self.common = w, seqs, new, heads, kv_heads, most // PAGE
        pages = self.common + seqs * (OWN // PAGE)
        codes = [torch.randint(-127, 128, (pages, kv_heads, PAGE, DIM), generator=g, device="cuda", dtype=torch.int8)
                 for _ in range(2)]
        # scores of some units, so that some tens of keys have most of the weight; values up to 1
        scales = [torch.empty((pages, kv_heads), device="cuda").uniform_(0.5 * s, s, generator=g) for s in (1 / 20, 1 / 127)]
        self.cache = w.KVCache(*codes, *scales)
        self.q = torch.randn((seqs * new, heads, DIM), generator=g, device="cuda").half()
        self.starts = torch.arange(0, seqs * new + 1, new, dtype=torch.int32, device="cuda")
        self.groups = torch.tensor([0, seqs], dtype=torch.int32, device="cuda")

    def tables(self, prefix):
        """Rows on the first `prefix` positions, their own pages behind these."""
        common = torch.arange(prefix // PAGE, dtype=torch.int32, device="cuda").expand(self.seqs, -1)
        own = self.common + torch.arange(self.seqs * (OWN // PAGE), dtype=torch.int32, device="cuda").view(self.seqs, -1)
        return (torch.cat([common, own], 1).contiguous(),
                torch.full((self.seqs,), prefix + OWN, dtype=torch.int32, device="cuda"))

    def call(self, prefix):
        """(result, the plan's words: whether the tensor-core kernel has the group, its SMs, the other kernel's)"""
        w = self.w
        table, lens = self.tables(prefix)
        ws = torch.zeros(w.w4a16_kv_attention_shared_workspace(self.heads, self.kv_heads, DIM, self.seqs, 1, self.seqs * self.new),
                         dtype=torch.uint8, device="cuda")
        out = w.w4a16_kv_attention_shared(self.q, self.cache, table, lens, self.starts, self.new, self.groups,
                                          torch.tensor([prefix], dtype=torch.int32, device="cuda"), workspace=ws)
        torch.cuda.synchronize()
        assert w.w4a16_last_device_error() == 0
        # the workspace begins with an entry of 32 bytes for each group and sequence, then 16 for the group
        at = (1 + self.seqs) * 32 + 16
        return out, ws[at:at + 12].view(torch.int32).tolist()

    def alone(self, prefix):
        table, lens = self.tables(prefix)
        return self.w.w4a16_kv_attention(self.q, self.cache, table, lens, self.starts, self.new)


# prefixes whose calls are estimated at 0.4 to 4.5 ms: the last two at more than 4
@pytest.mark.parametrize("seqs, new, heads, kv_heads, prefixes", [
    (512, 2, 64, 8, [8192, 65536, 98304, 114688, 117760, 122880, 131072]),
    (1024, 1, 128, 8, [8192, 32768, 53248, 56320, 59392, 65536]),
    (1024, 1, 64, 4, [16384, 65536, 114688, 118784, 122880, 131072]),
    (256, 16, 32, 32, [8192, 32768, 53248, 56320, 59392, 65536]),
])
def test_division(cuda_lib, seqs, new, heads, kv_heads, prefixes):
    p = Shared(cuda_lib, seqs, new, heads, kv_heads, prefixes[-1])
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    words = [p.call(n)[1] for n in prefixes]
    assert all(use == 1 for use, _, _ in words), words
    many = [k for _, k, _ in words]
    # (one kernel after the other, on all SMs, and side by side, on nine of ten, may be as good as one another)
    assert all(10 * b >= 9 * a for a, b in zip(many, many[1:])), words
    # side by side or one after the other, no SM without work
    assert all(k + rest == sms or k == rest == sms for _, k, rest in words), words
    assert many[-1] > sms // 2


def test_result_of_a_call_of_several_ms(cuda_lib):
    """Both ways of reading the keys are within the same bound of the exact result: outputs rounded once, weights that meet
    the values as fp16, 2^-11 of each, and 2^-12 for scores and exponentials; the values are below 1."""
    p = Shared(cuda_lib, 512, 2, 64, 8, 131072)
    out, want = p.call(131072)[0].double(), p.alone(131072).double()
    bound = 2 * (2.0 ** -11 + 2.0 ** -12) + 2.0 ** -11 * (out.abs() + want.abs())
    assert bool(((out - want).abs() <= bound).all())
    assert float(want.abs().max()) > 0.2                               # something to compare
