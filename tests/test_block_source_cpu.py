"""What the layer operators' sources state, checked without a GPU."""
import os
import re

from latent_projection_top_amd import block

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_cleared_part_of_a_workspace_matches_the_header():
    src = open(os.path.join(ROOT, "include", "block.h")).read()
    assert int(re.search(r"#define BLOCK_WORKSPACE_ZEROED (\d+)", src).group(1)) == block.WORKSPACE_ZEROED
