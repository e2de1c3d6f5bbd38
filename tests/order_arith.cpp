// The division of the order of rows into workgroups, for tests/test_order_plan_cpu.py: compiled with g++.
#include "order_plan.hpp"

extern "C" {

int order_is_small(int64_t S, int64_t G) { return g355::order_small(S, G); }
void order_division(int64_t S, int64_t G, int* chunk, int* chunks) { g355::order_chunks(S, G, *chunk, *chunks); }

}  // extern "C"
