"""Names of the repository's files can be checked out and listed anywhere.  No GPU needed."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_paths_are_plain():
    """No tracked path has blanks, quotes, colons, control characters or the like."""
    try:
        out = subprocess.run(["git", "-C", ROOT, "ls-files", "-z"], capture_output=True, check=True).stdout
    except (OSError, subprocess.CalledProcessError):
        pytest.skip("not a git checkout")
    paths = [p.decode() for p in out.split(b"\0") if p]
    assert paths
    plain = set("abcdefghijklmnopqrstuvwxyzABCDEFGHIJKLMNOPQRSTUVWXYZ0123456789._-/")
    assert [p for p in paths if set(p) - plain] == []
