"""Order between the warps of the chunk attention, read from its source (no GPU): what the
warp that goes over V finds in a piece (bad[]) is written before the softmax reads it.

The softmax waits for o_full, on which only the product warp arrives.  So the order has to
come through that warp: it waits for `clean` of the piece's last plane of V, on which the
value warp arrives after its store."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "block_diffusion_speculative_fuse_gb300", "csrc", "attention_chunk.cu")


def test_the_last_plane_of_every_piece_is_waited_for():
    text = open(SOURCE).read()
    found = re.findall(r"const int iv = take\(([^;]*)\);", text)
    assert len(found) == 1
    waits = found[0].replace("||", "or").replace("&&", "and")
    # (a piece all of whose keys every row sees has clean0 >= n)
    for n in (1, 2, 3, 7, 100):
        for clean0 in (-5, -1, 0, 1, n - 1, n, n + 1, n + 1000):
            assert eval(waits, {}, dict(c=n - 1, n=n, clean0=clean0)), (n, clean0)


def test_what_was_found_is_written_before_the_plane_is_handed_on():
    text = open(SOURCE).read()
    role = text[text.index("V's values\n"):]
    role = role[:role.index("piece_done()")]
    assert role.count("bad[taken % kPieces] = found") == role.count("mbar_arrive(&clean[st])") == 1
    assert role.index("bad[taken % kPieces] = found") < role.index("mbar_arrive(&clean[st])")
    # and only the product warp arrives on o_full, when it has issued the piece's products
    assert re.findall(r"mbar_init\(o_full, (\d+)\)", text) == ["2"]
    assert len(re.findall(r"mbar_arrive\(o_full\)|commit\(o_full\)", text)) == 2
