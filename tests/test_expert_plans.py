"""Which kernel a call's shape takes, and what the binding asks for it, on the host."""
import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from weight_only_int4_stats_b200 import build
    build.build()
    import weight_only_int4_stats_b200 as awq
    return awq.lib()


@pytest.mark.parametrize("N,K", [(14336, 4096), (4096, 14336), (37, 384)])
@pytest.mark.parametrize("bits", [4, 3])
def test_up_to_8_fp16_rows_with_inv_s_are_held_in_two_parts(L, N, K, bits):
    """The workspace of 1 to 8 rows holds two fp16 rows of each (the kernel that rounds nothing
    before the output); 9 rows need no such copy of fp16 activations."""
    def need(M):
        return L.awq_gemm_epilogue_workspace_size(M, N, K, bits, 1, 0)
    for M in range(1, 9):
        assert M * 4 * K <= need(M)
    splits = (need(9) + 256) // (9 * N * 4)   # partial sums of slices of K alone
    assert need(9) <= splits * 9 * N * 4 + 255
    for E in (2, 128):
        for T in (1, 4 * E, 4 * E + 1, 8 * E):
            assert L.awq_gemm_grouped_workspace_size(T, E, N, K, bits, 1, 0) >= T * 4 * K
        assert L.awq_gemm_grouped_workspace_size(8 * E + 1, E, N, K, bits, 1, 0) == 0


class Devices:
    """A machine of unlike GPUs: the library's size query goes by the current device."""

    def __init__(self, awq, monkeypatch):
        self.current, self.calls, self.allocated = 0, [], []
        monkeypatch.setattr(awq, "lib", lambda: self)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.current)
        monkeypatch.setattr(torch.cuda, "device", self.guard)
        monkeypatch.setattr(awq, "_current_raw_stream", lambda index: 0)
        monkeypatch.setattr(awq, "_new", self.new)

    def guard(self, index):
        class Guard:
            def __enter__(g):
                g.before, self.current = self.current, index

            def __exit__(g, *exc):
                self.current = g.before
        return Guard()

    def new(self, nbytes, dtype, index, stream):
        self.allocated.append((index, nbytes))

        class Memory:
            get_device, is_contiguous = (lambda m: index), (lambda m: True)
            data_ptr, numel, element_size = (lambda m: 256), (lambda m: nbytes), (lambda m: 1)
        return Memory()

    def awq_size(self, n):
        return n * (self.current + 1)

    def awq_op(self, x, ws, ws_bytes, stream):
        self.calls.append((self.current, x, ws_bytes))
        return 0 if ws_bytes >= x * (self.current + 1) else 3


def test_binding_plans_for_the_tensors_device(monkeypatch):
    import weight_only_int4_stats_b200 as awq
    box = Devices(awq, monkeypatch)
    for index in (1, 0, 1, 3):   # not the current device, and the same sizes on each
        awq._call("awq_op", index, None, ("awq_size", 100), None, (100,))
        assert box.allocated[-1] == (index, 100 * (index + 1))
        assert box.calls[-1] == (index, 100, 100 * (index + 1)) and box.current == 0


def test_plain_products_size_covers_bf16(L):
    """At 4 bits up to 8 rows an odd N (or an X too large for shared memory) goes to the tensor-core
    path with bf16 activations, as at 3 bits: the size is the same for both."""
    for M, N, K in ((1, 1000, 11008), (4, 1000, 11008), (8, 40, 4096), (8, 4096, 65536)):
        need = L.awq_gemm_workspace_size(M, N, K, 4)
        assert need == L.awq_gemm_workspace_size(M, N, K, 3) and need >= 2 * M * N * 4
    assert L.awq_gemm_workspace_size(8, 1008, 4096, 4) == 0
