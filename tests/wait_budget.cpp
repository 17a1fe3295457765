// wait_budget.cpp -- prints whether a wait of argv[1] ns has taken more than twice the budget argv[2].
#include <cstdio>
#include <cstdlib>

#include "fa_kvcache.h"

int main(int, char **argv) {
    std::puts(fa::twice_over(std::strtoull(argv[1], nullptr, 10), std::strtoll(argv[2], nullptr, 10)) ? "over" : "within");
}
