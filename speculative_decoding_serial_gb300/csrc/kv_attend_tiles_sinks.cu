// kv_attend_tiles_sinks.cu — attention of many rows with a window and first keys that stay visible behind it. 2 x 2048 tokens, window
// 1,024, 100 first keys: 136 us (75 GFLOP, 0.55 PFLOP/s), the window alone 128; 64 channels 104 and 96. An item has ten blocks, and the change from
// one to the next, some 10 us and 3.4 times a CTA, weighs more than in long items.
#include "kv_attend_tiles.cuh"

namespace whead_kv_impl {
template int launch_tiles<true>(const HostCache& h, const AttendArgs& a, int max_q);
}
