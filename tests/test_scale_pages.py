"""copy_pages of a quantised cache: what the scales' copy would refuse is refused
before the codes move."""
import pytest
import torch


def test_misaligned_scales_are_refused_before_the_codes_move(monkeypatch):
    from weight_streaming_expert_gb300 import cache as C
    moved = []
    monkeypatch.setattr(C, "_copy", lambda name, *a: moved.append(name))
    pools = [torch.zeros(2, 4, 16, 2, 64, dtype=torch.uint8) for _ in range(2)]
    i = torch.arange(2, dtype=torch.int32)
    room = torch.zeros(2 * 4 * 2 * 16 + 32, dtype=torch.uint8)
    at = -room.data_ptr() % 16
    scales = lambda offset: room[at + offset:at + offset + 256].view(2, 4, 2, 16)
    C.copy_pages(*pools, i[:1], i[1:], k_scale=scales(0), v_scale=scales(16))
    assert moved == ["moe_copy_pages"] * 2
    for bad in ((8, 0), (0, 4), (0, 1)):
        with pytest.raises(ValueError, match="16 bytes"):
            C.copy_pages(*pools, i[:1], i[1:], k_scale=scales(bad[0]), v_scale=scales(bad[1]))
    assert len(moved) == 2
