"""The items that kvq_attend_prompts cuts packed prompts into: never more than its
workspace holds, whatever starts holds (no GPU needed)."""
import os
import subprocess

from kv_cache_quantization_kvq_gb300 import builder

HERE = os.path.dirname(os.path.abspath(__file__))


def test_items_of_prompts(tmp_path):
    exe = str(tmp_path / "plan_check")
    subprocess.run([builder._nvcc(), "-O1", "-std=c++17", "-I", builder.CSRC, "-o", exe,
                    os.path.join(HERE, "cuda", "plan_check.cu")], check=True, capture_output=True, text=True, timeout=600)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout
