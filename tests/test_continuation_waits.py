"""A warp of the many-row attention kernel whose lanes vote again after a wait gives up as a whole at the time limit: a
lane that left alone would keep the others in the vote for good.  Two lanes of a warp that disagree at the limit cannot be
arranged in a test, so this reads the source; CPU only."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "joint_video_audio_rope_b200", "csrc")


def _roles():
    """The parts of the many-row kernel by the banner comment that opens them."""
    with open(os.path.join(CSRC, "cache_attn_tc.cu")) as f:
        text = f.read()
    parts = re.split(r"// -{20,} (\w[\w ]*)\n", text)
    return dict(zip(parts[1::2], parts[2::2]))


def test_the_roles_are_found():
    assert {"MMA issuer", "pages", "converters", "softmax", "epilogue", "teardown"} <= set(_roles())


def test_converters_and_the_page_warp_wait_as_warps():
    for role in ("converters", "pages"):
        text = _roles()[role]
        assert "all_wait(" in text
        assert not re.search(r"(?<!\w)wait_for\(", text), role
