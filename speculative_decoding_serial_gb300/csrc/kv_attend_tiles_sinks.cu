// kv_attend_tiles_sinks.cu — attention of many rows with a window and first keys that stay visible behind it.
#include "kv_attend_tiles.cuh"

namespace whead_kv_impl {
template int launch_tiles<true>(const HostCache& h, const AttendArgs& a, int max_q);
}
