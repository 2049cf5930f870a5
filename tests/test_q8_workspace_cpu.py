"""The layer's workspaces hold what the layer's own calls need: the calls on 8-bit rows live in
regions that they leave idle, and add room only where sums go in parts."""
import pytest


@pytest.fixture(scope="module")
def sm():
    from sparse_mixture_experts_switch_b200 import build
    build.build()
    from sparse_mixture_experts_switch_b200 import switch_moe
    return switch_moe


# the layer's regions alone, forward and backward
LAYER = [((32768, 1024, 4096, 128, 1.0), 0, 421449728, 785176576),
         ((65536, 4096, 10240, 64, 1.25), 0, 3040227328, 4851775488),
         ((700, 320, 832, 6, 1.25), 0, 2684928, 4887552),
         ((8000, 128, 192, 3, 2.0), 0, 14672896, 27676672),
         ((400, 128, 320, 5, 1.0), 512, 984064, 2322432)]


@pytest.mark.parametrize("sizes,flags,forward,backward", LAYER)
def test_no_bytes_for_the_8_bit_calls(sm, sizes, flags, forward, backward):
    cfg = sm.config(*sizes, flags=flags)
    assert sm.switch_workspace_size(cfg) == forward
    assert sm.switch_backward_workspace_size(cfg) == backward


# few tiles and long sums: (sizes, the layer's regions alone forward and backward)
FEW = [((300, 64, 4672, 1, 1.0), 2915328, 5991424), ((20, 5632, 5696, 1, 1.0), 1775616, 3515392),
       ((90, 128, 9472, 3, 4.0), 7046144, 14243840), ((3, 64, 9728, 8, 8.0), 500736, 1017856)]


@pytest.mark.parametrize("sizes,forward,backward", FEW)
def test_room_for_parts_is_bounded(sm, sizes, forward, backward):
    cfg = sm.config(*sizes)
    f, b = sm.switch_workspace_size(cfg), sm.switch_backward_workspace_size(cfg)
    assert forward < f <= forward + (24 << 20) and backward <= b <= backward + (24 << 20) and f <= b
