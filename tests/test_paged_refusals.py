"""Pointers that the paged calls' kernels could not read without a fault are
refused on the host (no GPU needed: every call is refused, or stopped by the
test hook, before it launches)."""
import pytest

from test_paged_abi import FAKE, append_args, attend_args, paged, plan_args, rope_args  # noqa: F401


@pytest.fixture(autouse=True)
def stop_at_the_launch(monkeypatch):
    monkeypatch.setenv("QWM_FAULT_INJECT", "launch")


def moved(pack, paged, at, by):
    """The packed arguments with `by` added to 64-bit field `at`."""
    raw = bytearray(pack)
    raw[8 * at: 8 * at + 8] = (int.from_bytes(raw[8 * at: 8 * at + 8], "little") + by).to_bytes(8, "little")
    return bytes(raw)


@pytest.mark.parametrize("by,status", [(1, 1), (2, 1), (3, 1), (4, 6)])
def test_words_off_their_boundary(paged, by, status):  # noqa: F811
    L = paged.lib()
    # plan: 64-bit slots (field 8) need 8 bytes
    plan = plan_args(paged)
    for at in range(11):
        assert L.qwm_paged_plan(moved(plan, paged, at, by), None) == (1 if at == 8 else status), at
    release = paged._RELEASE.pack(*[FAKE] * 6, 5, 3, 4, 16)
    for at in range(6):
        assert L.qwm_paged_release(moved(release, paged, at, by), None) == status, at
    rope = rope_args(paged, status=FAKE)
    for at in (15, 16):   # positions, status
        assert L.qwm_qk_norm_rope(moved(rope, paged, at, by), None) == status, at
    assert L.qwm_paged_append(append_args(paged, status=FAKE + by), None) == status
    for name in ("lse", "table", "lens", "cu", "status"):
        assert L.qwm_paged_attend(attend_args(paged, **{name: FAKE + by}), None) == status, name


@pytest.mark.parametrize("max_new", [33, 1 << 31, 1 << 61, (1 << 63) - 1])
def test_kernel_choice_of_long_hints(paged, max_new):  # noqa: F811
    """The hint times the head group does not leave 64 bits."""
    for heads, kv_heads in ((1, 1), (8, 1), (8, 2), (48, 3)):
        assert paged.lib().qwm_paged_attend_kernel_for(1, heads, kv_heads, max_new) == 3
