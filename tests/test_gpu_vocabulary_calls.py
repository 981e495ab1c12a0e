"""The losses and the embedding called from several threads, and from graphs that
share a stream's workspace with calls that outgrow it."""
import threading

import pytest

import trellis_coded_bit_prefill_amd as tp
from tests.test_gpu_vocabulary_run import EXTRA, K, N, need_gpu, parts  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def losses(p, x):
    return (*tp.cross_entropy(x, *p["packed"], p["target"], keep=True),
            *tp.distill(x, *p["packed"], p["index"], p["logits"], temperature=2.0, keep=True))


def embedding(p, x):
    codes, scales, bits = p["packed"]
    return (tp.embed(p["tokens"], codes, scales, K, bits, scale=3.0, extra=p["extra"]),
            tp.embed_backward(x, p["tokens"], N, EXTRA, scale=0.5))


def equal(got, want):
    import torch

    return len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("own_streams", [True, False])
def test_threads(parts, own_streams):  # noqa: F811
    """Four threads, each on a stream of its own or all on one, the same calls in other orders."""
    import torch

    print(f"threads, own streams {own_streams}", flush=True)
    p, x = parts, parts["x"]
    want = losses(p, x), embedding(p, x)
    torch.cuda.synchronize()
    one = torch.cuda.Stream()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream() if own_streams else one):
                for rep in range(8):
                    order = (0, 1) if (i + rep) % 2 else (1, 0)
                    got = [None, None]
                    for o in order:
                        got[o] = (losses, embedding)[o](p, x)
                    torch.cuda.current_stream().synchronize()
                    if not all(equal(a, b) for a, b in zip(got, want)):
                        wrong.append((i, rep))
        except Exception as e:  # (of this thread)
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("path", [None, False, True], ids=["auto", "few", "many"])
def test_two_graphs_and_calls_that_outgrow_their_workspace(parts, path):  # noqa: F811
    """Two graphs of one stream, replayed in turn with eager calls between them, the last ones of which need a larger
    workspace: the graphs go on in the old one."""
    import torch

    print(f"two graphs {path}", flush=True)
    p = parts
    x = p["x"].clone()
    stream = torch.cuda.Stream()
    tp.force_path(path)
    try:
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            losses(p, x), embedding(p, x)
        torch.cuda.synchronize()
        graphs = []
        for calls in (losses, embedding):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                outs = calls(p, x)
            graphs.append((graph, calls, outs))
        big = p["x"].repeat(40, 1)
        tokens, target = p["tokens"].repeat(40), p["target"].repeat(40)
        for rep in range(4):
            x.copy_(p["x"].roll(rep, 0))
            torch.cuda.synchronize()
            for graph, calls, outs in graphs + graphs[::-1]:
                for o in outs:
                    o.fill_(float("nan"))
                torch.cuda.synchronize()
                with torch.cuda.stream(stream):
                    graph.replay()
                    torch.cuda.current_stream().synchronize()
                    got = [o.clone() for o in outs]
                    want = calls(p, x)
                    if rep >= 1:
                        tp.cross_entropy(big, *p["packed"], target, keep=True)
                        tp.embed_backward(big, tokens, N, EXTRA)
                torch.cuda.synchronize()
                assert equal(got, want), (rep, calls.__name__)
    finally:
        tp.force_path(None)
