"""The tile shape asked for by gs_layer_tile decides the plan, without a GPU: partial sums of a
split contraction are as many as the shape's tiles leave room for.  Of the calling thread only."""
import threading


def test_tile_decides_the_plan():
    from differentiable_rasterizer_gb300 import abi, build
    build.build()

    def scratch():   # a plain sum of few tiles over 5000 k: split
        return abi.layer_ws_bytes("gs_linear", abi.linear_args(300, 5000, 200, 4096, 5000, 4096, 5000, 0, 0, 0, 0, 0, 4096, 200, 0,
                                                               0, abi.GS_BF16, abi.GS_BF16, abi.GS_BF16, 0))

    chosen, other = scratch(), []
    sizes = []
    try:
        for tile in range(4):
            abi.gs_layer_tile(tile)
            sizes.append(scratch())
        t = threading.Thread(target=lambda: other.append(scratch()))
        t.start()
        t.join()
    finally:
        abi.gs_layer_tile(-1)
    assert scratch() == chosen and other == [chosen]
    assert len(set(sizes)) > 1 and chosen in sizes
    part = 300 * 200 * 4
    assert all(s // part >= 2 for s in sizes)
