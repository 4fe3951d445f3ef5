"""The block manager's batched calls when the host runs out of memory."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_out_of_host_memory_changes_nothing(tmp_path):
    """Every allocation of pa_bm_append_chunks and pa_bm_keep fails in turn
    (tests/block_manager_oom.cpp): a refused call has changed nothing, one that went on has done
    its work, and no block is lost."""
    exe = str(tmp_path / "oom")
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17",
                    "-I", os.path.join(ROOT, "include"), "-o", exe,
                    os.path.join(ROOT, "tests", "block_manager_oom.cpp"),
                    os.path.join(ROOT, "paged_kv_cache_410_b200", "csrc", "pa_block_manager.cpp")],
                   check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
