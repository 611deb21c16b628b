"""The bench line's DRAM traffic is read from a record that names the attention source it was
measured on: the record has to be of the source as it stands."""
import bench


def test_the_record_is_of_the_current_attention_source():
    assert bench.read_traffic() is not None, bench.attn_source_hash()
