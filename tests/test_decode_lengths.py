"""The decode step refuses sequences that complete no entry (host logic, no GPU)."""
import pytest

from serving_lightning_indexer_gb300.decode_step import DecodeStep


@pytest.mark.parametrize("lengths,layers,need", [
    ([64, 1, 7], (2, 20), 2), ([0], (20,), 1), ([5, 0], (8, 9), 2), ([-3, 4], (20, 24), 1), ([1], tuple(range(2, 40)), 2),
    ([], (20,), 1),
])
def test_decode_step_refuses_a_sequence_without_an_entry(lengths, layers, need):
    """Such a sequence has no newest entry: its slot and the later sequences' would be others'."""
    with pytest.raises(ValueError, match=f"needs {need} tokens"):
        DecodeStep(lengths, seed=1, device="cpu", layers=layers)


@pytest.mark.parametrize("lengths,layers", [([2, 9], (2, 20)), ([1], (20, 21))])
def test_decode_step_takes_the_shortest_sequences(lengths, layers):
    """They pass the check and reach the calls, which take CUDA tensors only."""
    with pytest.raises(ValueError, match="CUDA tensors"):
        DecodeStep(lengths, seed=1, device="cpu", layers=layers)
