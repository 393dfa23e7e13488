// kv_attend_sinks.cu — attention of few rows with a window and first keys that stay visible behind it.
#include "kv_attend_rows.cuh"

namespace whead_kv_impl {
template int launch_few<true>(const HostCache& h, const AttendArgs& a, int max_q, int tile);
}
