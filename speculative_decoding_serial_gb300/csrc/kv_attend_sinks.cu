// kv_attend_sinks.cu — attention of few rows with a window and first keys that stay visible behind it: softmax over j < sinks and
// p - window < j <= p. The units between are left out of an item, so that the first keys cost one unit more. 32 sequences of 2,000 to 32,768
// keys, window 4,096, 4 first keys: 40.8 us (151 MB, 3.7 TB/s), the window alone 38.7; one on 20,001, window 1,024: 10.3 us, latency.
#include "kv_attend_rows.cuh"

namespace whead_kv_impl {
template int launch_few<true>(const HostCache& h, const AttendArgs& a, int max_q, int tile);
}
