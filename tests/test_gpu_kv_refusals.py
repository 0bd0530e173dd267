"""Arguments of the paged cache's calls that no tensor check sees: every wrong one is an HQArgError or an HQError, and
nothing is launched."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _calls(lib):
    """Right calls of the three operators, each as a function of what is changed."""
    c = lib.make_kv_cache("e4m3", 3, 16, 2, 64)
    bf, i32, i64 = torch.bfloat16, torch.int32, torch.int64
    z = lambda *s, dt: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    write = dict(qkv=z(3, 8 * 64, dt=bf), slots=z(3, dt=i64) - 1, num_q_heads=4)
    read = dict(page_table=z(1, 2, dt=i32), starts=z(2, dt=i64), total=4)
    attend = dict(q=z(2, 8, 64, dt=bf), page_table=z(2, 2, dt=i32), lens=z(2, dt=i32))
    return (lambda **k: lib.kv_write(c, **{**write, **k}), lambda **k: lib.kv_read(c, **{**read, **k}),
            lambda **k: lib.paged_attention(c, **{**attend, **k}))


def test_a_workspace_that_is_no_device_tensor(lib):
    for call in _calls(lib):
        for ws in (0, "workspace", 1 << 20, torch.zeros(1 << 20, dtype=torch.uint8),
                   torch.zeros(1 << 16, 4, dtype=torch.uint8, device="cuda")[:, :2]):
            with pytest.raises(lib.HQArgError):
                call(workspace=ws)
        call()
    torch.cuda.synchronize()


def test_numbers_past_their_fields(lib):
    """What a field cannot hold is refused by the binding, what is infinite in fp32 by the library."""
    write, read, attend = _calls(lib)
    for call, over in ((write, dict(eps="small")), (write, dict(eps=None)), (attend, dict(softcap=None)),
                       (attend, dict(scale="half")), (attend, dict(window=1 << 63)), (attend, dict(window=-(1 << 70))),
                       (attend, dict(window=1.5)), (attend, dict(window=None)), (read, dict(total=-1))):
        with pytest.raises(lib.HQArgError):
            call(**over)
    for call, over in ((write, dict(eps=1e39)), (write, dict(eps=float("inf"))), (attend, dict(scale=1e300)),
                       (attend, dict(scale=-1e39)), (attend, dict(softcap=1e39)), (attend, dict(window=-1))):
        with pytest.raises(lib.HQError) as e:
            call(**over)
        assert e.value.code == lib.HQ_ERR_INVALID_ARG
