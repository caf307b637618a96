"""What the grouped products' wrappers refuse on the host: operands whose
memory is not what the kernels read (no GPU, nothing is enqueued)."""
import pytest
import torch


@pytest.fixture(scope="module")
def F():
    import fp4_quantization_amd as F
    return F


def call(F, which, change, name):
    """A product of E = 3 segments whose operand `which` has one changed tensor."""
    E, R, N, K = 3, 32, 16, 64
    off = torch.tensor([0, 16, 16, 32])
    if name == "nt":
        a, b, c = F.alloc_layout(R, K, 0, E, "cpu"), F.alloc_layout(E * N, K, 0, E, "cpu"), torch.zeros(R, N)
    else:
        a, b, c = F.alloc_layout(N, R, 0, E, "cpu"), F.alloc_layout(K, R, 0, E, "cpu"), torch.zeros(E, N, K)
    change((a, b)[which])
    if name == "nt":
        F.ufp4_gemm_grouped_nt(F.config(), a, b, 0, off, K, c)
    else:
        F.ufp4_gemm_grouped_dw(F.config(), a, b, off, c)


def one_scale_for_all(q):
    q.tensor_scale = torch.ones(1).expand(3)


def every_second_scale(q):
    q.tensor_scale = torch.ones(6)[::2]


def wide_codes(q):
    q.codes = q.codes.to(torch.int16)


def float_scales(q):
    q.scales = q.scales.float()


@pytest.mark.parametrize("name", ["nt", "dw"])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("change", [one_scale_for_all, every_second_scale, wide_codes, float_scales])
def test_refused(F, name, which, change):
    with pytest.raises(ValueError, match="must h"):
        call(F, which, change, name)


@pytest.mark.parametrize("name", ["nt", "dw"])
def test_other_one_byte_types_pass_the_checks(F, name, monkeypatch):
    """Codes and scales are bytes whatever their type is called."""
    done = []
    monkeypatch.setattr(F.lib, "ufp4_gemm_grouped_nt", lambda *a: done.append(a) or 0)
    monkeypatch.setattr(F.lib, "ufp4_gemm_grouped_dw", lambda *a: done.append(a) or 0)
    monkeypatch.setattr(F, "_stream", lambda s: 0)

    def change(q):
        q.codes, q.scales = q.codes.view(torch.int8), q.scales.view(torch.float8_e4m3fn)

    call(F, 0, change, name)
    assert len(done) == 1
