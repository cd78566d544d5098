"""The package's names: `import *` needs no torch, the operators come by name."""
import subprocess
import sys

from conftest import ROOT


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_import_star_without_torch():
    r = run("import sys; sys.modules['torch'] = None\n"
            "from parity_binade_chunked_gb300 import *\n"
            "assert callable(seqsum_f64) and callable(version) and SeqsumPlan and issubclass(SeqsumError, RuntimeError)")
    assert r.returncode == 0, r.stderr


def test_import_star_does_not_load_torch():
    r = run("import sys\nfrom parity_binade_chunked_gb300 import *\nassert 'torch' not in sys.modules")
    assert r.returncode == 0, r.stderr


def test_operators_by_name():
    r = run("import parity_binade_chunked_gb300 as sq\n"
            "names = ['sample_tokens', 'token_logprob', 'token_logprob_grad', 'token_logprob_backward', 'TensorList']\n"
            "assert set(names) <= set(dir(sq)) and set(sq.__all__) <= set(dir(sq))\n"
            "from parity_binade_chunked_gb300 import sample_tokens, TensorList\n"
            "assert all(callable(getattr(sq, n)) for n in names)\n"
            "assert not hasattr(sq, 'no_such_name')")
    assert r.returncode == 0, r.stderr
